"""Convenience wrappers over the sequence operators: 4-bit pointwise layers, blocks with carried states
(a selective scan or a gated delta rule), beam search, and the verification of drafted tokens.  Shapes,
types and strides are checked here; the computation runs in the library's kernels.

A block is  in-projection -> causal depthwise layer -> (step, B, C) projection -> selective scan
gated by the in-projection's other half -> out-projection:

    block = StateSpaceBlock(..., slots=16)
    y = block.prompt(x, cu, slots)        # packed prompts [tokens, dim]
    y = block.step(x, slots)              # one token of each sequence [batch, dim]

(:class:`DeltaRuleBlock` has the same calls.)  Tokens that a smaller model has drafted are checked a
whole row of them at a time, in slots of their own, and the states then moved on over those that stand:

    verify = DraftVerifier(requests, drafts, vocab)
    for p in pools: p[spare] = p[slots]          # int64 slots
    logits = model(rows, cu, spare, carry)       # each request's last token and its drafts
    accepted, following = verify(logits, tokens, draft_logits)
    model(rows, *verify.kept(accepted, slots), carry)

Every call works on torch's current stream.  With ``stream`` (a torch stream or a raw handle) all of
it, the projections and what it allocates among it, works on that stream instead, behind what the
current stream holds at the call; whoever uses the results or the states on another stream waits for it.
(What makes a layer's weights, and ``weight`` that shows them, take no ``stream``.)
"""
from __future__ import annotations

from typing import Optional, Sequence

import torch

from . import (ACT_CODES, beam_problem, delta_problem, draft_problem, dw1d_problem, fcm_beam_reorder,
               fcm_beam_select, fcm_beam_workspace, fcm_delta_fwd, fcm_delta_step, fcm_delta_workspace,
               fcm_draft_verify, fcm_draft_workspace, fcm_dw1d_fwd, fcm_dw1d_step, fcm_mx4_dequantize,
               fcm_mx4_fwd, fcm_mx4_quantize, fcm_mx4x4_fwd, fcm_q4_fwd, fcm_scan_fwd, fcm_scan_step,
               fcm_scan_workspace, mx4_problem, q4_problem, scan_problem)

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


def quantize_mx4(x: torch.Tensor, stream=None):
    """Codes [rows, C/2] and scales [rows, C/32], uint8, of [rows, C] values in blocks of 32 channels: a
    power of two for the block, and for each channel the nearest of 0, 0.5, 1, 1.5, 2, 3, 4 and 6 with a
    sign.  A value below the block's largest code is off by at most a quarter of itself or a quarter of
    the scale, whichever is larger."""
    if stream is not None:
        return _on(stream, lambda: quantize_mx4(x), x)
    _need(x.dtype in DTYPE_NAMES, "x must be float32, float16 or bfloat16")
    _need(_on_gpu(x), "x must be on the current GPU")
    _need(x.dim() == 2 and x.shape[1] > 0 and x.shape[1] % 32 == 0, "x must be [rows, C], C a multiple of 32")
    rows, C = x.shape
    x = _rows(x, C, x.dtype, "x", x.device)
    q = torch.empty(rows, C // 2, dtype=torch.uint8, device=x.device)
    scales = torch.empty(rows, C // 32, dtype=torch.uint8, device=x.device)
    fcm_mx4_quantize(mx4_problem(DTYPE_NAMES[x.dtype], rows, C, 1, ldx=_stride(x)), x, q, scales)
    return q, scales


class MX4Linear:
    """y = act(x W^T + bias) with W in microscaled 4-bit floating point: q [K, C/2] and scales [K, C/32],
    uint8 (see :func:`quantize_mx4`), bias [K] float32 or None; activations of `dtype`.  With
    `quantize_input` x goes into the same codes first and the product runs on the scaled matrix
    instructions, for prompts of any length; without, it is meant for a few tokens (the weights are read
    and converted again for every 32: 4096 -> 8192 channels take 13 us for 64 tokens, 1153 for 8192, with
    `quantize_input` 12 and 207)."""

    def __init__(self, q, scales, bias=None, act: str = "none", dtype: torch.dtype = torch.bfloat16,
                 quantize_input: bool = False):
        _need(q.dim() == 2 and q.dtype == torch.uint8 and q.is_contiguous() and q.shape[1] > 0 and
              q.shape[1] % 16 == 0, "q must be [K, C/2] uint8, C a multiple of 32")
        self.K, self.C = q.shape[0], q.shape[1] * 2
        _need(scales.dtype == torch.uint8 and scales.is_contiguous() and
              tuple(scales.shape) == (self.K, self.C // 32), f"scales must be [{self.K}, {self.C // 32}] uint8")
        _need(bias is None or (bias.dtype == torch.float32 and tuple(bias.shape) == (self.K,) and
                               bias.is_contiguous()), f"bias must be [{self.K}] float32")
        for name, v in (("scales", scales), ("bias", bias)):
            if v is not None:
                _beside(v, q.device, name)
        _need(act in ACT_CODES, f"act must be one of {sorted(ACT_CODES)}")
        _need(dtype in (torch.float16, torch.bfloat16), "dtype must be float16 or bfloat16")
        self.q, self.scales, self.bias = q, scales, bias
        self.act, self.dtype, self.quantize_input = act, dtype, quantize_input

    @classmethod
    def from_weight(cls, weight, bias=None, act: str = "none", dtype: Optional[torch.dtype] = None,
                    quantize_input: bool = False) -> "MX4Linear":
        """Of a [K, C] weight on the GPU; dtype: the weight's if it is a 16-bit one, else bfloat16."""
        if dtype is None:
            dtype = weight.dtype if weight.dtype == torch.float16 else torch.bfloat16
        return cls(*quantize_mx4(weight), bias=bias, act=act, dtype=dtype, quantize_input=quantize_input)

    def weight(self) -> torch.Tensor:
        """The [K, C] weight the codes stand for, in float32."""
        _need(_on_gpu(self.q), "the weights must be on the current GPU")
        w = torch.empty(self.K, self.C, device=self.q.device)
        fcm_mx4_dequantize(mx4_problem("f32", self.K, self.C, 1), self.q, self.scales, w)
        return w

    def __call__(self, x, out=None, stream=None) -> torch.Tensor:
        if stream is not None:
            return _on(stream, lambda: self(x, out), x, out)
        _need(_on_gpu(self.q), "the weights must be on the current GPU")
        x = _rows(x, self.C, self.dtype, "x", self.q.device)
        M = x.shape[0]
        if out is None:
            out = torch.empty(M, self.K, dtype=self.dtype, device=x.device)
        else:
            _out(out, M, self.K, self.dtype, x.device)
        name = DTYPE_NAMES[self.dtype]
        if self.quantize_input:
            xq, xs = quantize_mx4(x)
            fcm_mx4x4_fwd(mx4_problem(name, M, self.C, self.K, self.act, ldy=_stride(out)), xq, xs, self.q,
                          self.scales, self.bias, out)
            return out
        if x.data_ptr() % 16 or _stride(x) % 8:
            x = x.clone(memory_format=torch.contiguous_format)
        fcm_mx4_fwd(mx4_problem(name, M, self.C, self.K, self.act, ldx=_stride(x), ldy=_stride(out)), x, self.q,
                    self.scales, self.bias, out)
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


class DeltaRuleBlock:
    """A block of the gated delta rule and the states of `slots` sequences:  in-projection -> causal
    depthwise layer with SiLU on queries, keys and values -> delta rule, its output normalised and gated
    -> out-projection.  Hv value heads of Dv channels, Hk key heads of Dk (Hv a multiple of Hk).

    in_proj: dim -> 2*Hk*Dk + 2*Hv*Dv + 2*Hv (queries, keys, values, gate, step, strength); conv_w
    [2*Hk*Dk + Hv*Dv, W], conv_b the same in float32 or None; A [Hv] float32, negative; dt_bias [Hv]
    float32 or None; norm [Dv] float32 or None; out_proj: Hv*Dv -> dim.  The projections are callables on
    [rows, channels] such as :class:`MX4Linear`."""

    def __init__(self, in_proj, conv_w, conv_b, A, dt_bias, norm, out_proj, Hk: int, Dk: int, Dv: int, slots: int,
                 scale: float = 0.0, eps: float = 1e-6):
        self.Hk, self.Hv, self.Dk, self.Dv = Hk, A.shape[0], Dk, Dv
        self.keys, self.inner = Hk * Dk, A.shape[0] * Dv
        self.mixed = 2 * self.keys + self.inner
        _need(conv_w.dtype in DTYPE_NAMES, "conv_w must be float32, float16 or bfloat16")
        _need(conv_w.dim() == 2 and conv_w.shape[0] == self.mixed, f"conv_w must be [{self.mixed}, W]")
        _need(Hk > 0 and self.Hv % Hk == 0, "the value heads must be a multiple of the key heads")
        for name, v, n in (("A", A, self.Hv), ("conv_b", conv_b, self.mixed), ("dt_bias", dt_bias, self.Hv),
                           ("norm", norm, Dv)):
            if v is not None:
                _need(tuple(v.shape) == (n,) and v.dtype == torch.float32 and v.is_contiguous(),
                      f"{name} must be [{n}] float32")
                _beside(v, conv_w.device, name)
        self.in_proj, self.out_proj = in_proj, out_proj
        self.conv_w, self.conv_b, self.A, self.dt_bias, self.norm = conv_w.contiguous(), conv_b, A, dt_bias, norm
        self.W, self.slots, self.scale, self.eps = conv_w.shape[1], slots, scale, eps
        self.dtype, self.name = conv_w.dtype, DTYPE_NAMES[conv_w.dtype]
        self.window = torch.zeros(slots, self.W - 1, self.mixed, dtype=self.dtype, device=conv_w.device)
        self.state = torch.zeros(slots, self.Hv, Dk, Dv, device=conv_w.device)

    _projected = StateSpaceBlock._projected
    _index = StateSpaceBlock._index

    def _parts(self, x):
        """(queries, keys and values together, gate, step, strength): the in-projection's parts."""
        p = self._projected(self.in_proj(x), x.shape[0], self.mixed + self.inner + 2 * self.Hv, "in_proj's result")
        at = self.mixed + self.inner
        return p[:, :self.mixed], p[:, self.mixed:at], p[:, at:at + self.Hv], p[:, at + self.Hv:]

    def _conv(self, xs, seqs: int):
        return dw1d_problem(self.name, self.mixed, self.W, tokens=xs.shape[0], seqs=seqs, slots=self.slots,
                            ldx=_stride(xs))

    def _rule(self, u, z, a, b, seqs: int):
        """The rule's problem and its inputs: u's parts, and those beside it."""
        prob = delta_problem(self.name, self.Hk, self.Hv, self.Dk, self.Dv, tokens=u.shape[0], seqs=seqs,
                             slots=self.slots, scale=self.scale, eps=self.eps, ldq=_stride(u), ldk=_stride(u),
                             ldv=_stride(u), lda=_stride(a), ldb=_stride(b), ldz=_stride(z))
        return prob, (u[:, :self.keys], u[:, self.keys:2 * self.keys], u[:, 2 * self.keys:], a, b, self.A,
                      self.dt_bias, self.norm, z)

    def prompt(self, x, cu, slots, carry=None, stream=None) -> torch.Tensor:
        """x: [tokens, dim], sequence b in rows cu[b] .. cu[b+1]-1 and state slot slots[b]; with
        carry[b] != 0 it continues from there."""
        if stream is not None:
            return _on(stream, lambda: self.prompt(x, cu, slots, carry), x, cu, slots, carry)
        _need(_on_gpu(self.window), "the block must be on the current GPU")
        T, B, dev = x.shape[0], slots.shape[0], self.window.device
        self._index(cu, B + 1, "cu")
        self._index(slots, B, "slots")
        self._index(carry, B, "carry")
        xs, z, a, b = self._parts(x)
        u = torch.empty(T, self.mixed, dtype=self.dtype, device=dev)
        fcm_dw1d_fwd(self._conv(xs, B), xs, self.conv_w, self.conv_b, cu, slots, carry, self.window, u)
        prob, parts = self._rule(u, z, a, b, B)
        y = torch.empty(T, self.inner, dtype=self.dtype, device=dev)
        ws = torch.empty(max(16, fcm_delta_workspace(prob)), dtype=torch.uint8, device=dev)
        fcm_delta_fwd(prob, *parts, cu, slots, carry, self.state, ws, y)
        return self.out_proj(y)

    def step(self, x, slots, stream=None) -> torch.Tensor:
        """x: [batch, dim], one token of the sequence in slots[b] (outside [0, slots): an idle row)."""
        if stream is not None:
            return _on(stream, lambda: self.step(x, slots), x, slots)
        _need(_on_gpu(self.window), "the block must be on the current GPU")
        B, dev = x.shape[0], self.window.device
        self._index(slots, B, "slots")
        xs, z, a, b = self._parts(x)
        u = torch.empty(B, self.mixed, dtype=self.dtype, device=dev)
        fcm_dw1d_step(self._conv(xs, B), xs, self.conv_w, self.conv_b, slots, self.window, u)
        prob, parts = self._rule(u, z, a, b, B)
        y = torch.empty(B, self.inner, dtype=self.dtype, device=dev)
        fcm_delta_step(prob, *parts, slots, self.state, y)
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


class DraftVerifier:
    """Verification of up to `drafts` drafted tokens of each of `requests` requests: tokens drawn this way
    are distributed as the target model's alone.  temperature 0: the largest logit alone counts."""

    def __init__(self, requests: int, drafts: int, vocab: int, temperature: float = 1.0):
        _need(requests >= 0 and drafts >= 1 and vocab >= 1, "sizes must be positive")
        self.requests, self.drafts, self.vocab, self.temperature = requests, drafts, vocab, temperature

    def _ints(self, t, n: int, name: str, device):
        _beside(t, device, name)
        _need(t.dtype == torch.int32 and t.numel() == n and t.is_contiguous(), f"{name} must have {n} int32 values")

    def __call__(self, target, tokens, draft=None, counts=None, uniform=None, stream=None):
        """target: logits [requests*(drafts+1), vocab] of the target model after a request's last token and
        after each of its drafts; tokens: [requests, drafts] int32; draft: logits [requests*drafts, vocab]
        that the tokens were drawn from (None: they were picked, with probability 1); counts: [requests]
        int32, how many of its tokens a request uses (None: all); uniform: [requests*(drafts+1)] float32 in
        [0, 1) (None: drawn here).  Returns (accepted, following), [requests] int32: how many tokens stand and
        the one behind them, -1 behind a row without any finite logit."""
        if stream is not None:
            return _on(stream, lambda: self(target, tokens, draft, counts, uniform), target, tokens, draft, counts,
                       uniform)
        R, D, V = self.requests, self.drafts, self.vocab
        _need(target.dtype in DTYPE_NAMES, "target must be float32, float16 or bfloat16")
        _need(_on_gpu(target), "target must be on the current GPU")
        dev = target.device
        target = _rows(target, V, target.dtype, "target", dev)
        _need(target.shape[0] == R * (D + 1), f"target must have {R * (D + 1)} rows")
        if draft is not None:
            draft = _rows(draft, V, target.dtype, "draft", dev)
            _need(draft.shape[0] == R * D, f"draft must have {R * D} rows")
        self._ints(tokens, R * D, "tokens", dev)
        if counts is not None:
            self._ints(counts, R, "counts", dev)
        if uniform is None and self.temperature != 0:
            uniform = torch.rand(R * (D + 1), device=dev)
        if uniform is not None:
            _beside(uniform, dev, "uniform")
            _need(uniform.dtype == torch.float32 and uniform.numel() == R * (D + 1) and uniform.is_contiguous(),
                  f"uniform must have {R * (D + 1)} float32 values")
        prob = draft_problem(DTYPE_NAMES[target.dtype], R, D, V, self.temperature, ldt=_stride(target),
                             ldd=0 if draft is None else _stride(draft))
        ws = torch.empty(max(16, fcm_draft_workspace(prob)), dtype=torch.uint8, device=dev)
        accepted = torch.empty(R, dtype=torch.int32, device=dev)
        following = torch.empty(R, dtype=torch.int32, device=dev)
        fcm_draft_verify(prob, target, draft, tokens, counts, uniform, ws, accepted, following)
        return accepted, following

    def kept(self, accepted, slots, stream=None):
        """(cu, slots) of 2*requests sequences for a block's ``prompt`` over the verified rows, each request's
        last token and its drafts: the rows that stand move the state in the request's slot on, the rows
        behind them belong to no slot.  (A caller's carry has 2*requests values.)  The states are bit for bit those
        that the rows gave when they were verified if a request has at most 16, else within their rounding."""
        if stream is not None:
            return _on(stream, lambda: self.kept(accepted, slots), accepted, slots)
        R, D = self.requests, self.drafts
        self._ints(accepted, R, "accepted", accepted.device)
        self._ints(slots, R, "slots", accepted.device)
        first = torch.arange(0, R * (D + 1), D + 1, dtype=torch.int32, device=accepted.device)
        cu = torch.empty(2 * R + 1, dtype=torch.int32, device=accepted.device)
        cu[0:-1:2], cu[1::2] = first, first + accepted + 1
        cu[-1:].fill_(R * (D + 1))
        return cu, torch.stack([slots, torch.full_like(slots, -1)], 1).reshape(-1)
