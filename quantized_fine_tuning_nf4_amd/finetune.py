"""What sits around the QLoRA linear in a fine-tuning step, and in serving
the tuned model: activation checkpoints in 8 bits with the linear's backward
from them, the norms before and after a block fused with its gate and residual
scale, and the log probabilities of given tokens with their gradient.

As in the package's other calls, the functions carry the C names and only
check and marshal arguments; outputs and workspaces are torch allocations on
the current stream.

    h, y, x8 = block_norm_fwd(h, w_pre, o=o, w_post=w_post, gate=g, scale=a, pack=True)
    dX, dA, dB = qlora_linear_bwd_act8(st, x8, dY, A, B, alpha, u)
    r = token_logprobs_fwd(logits, targets, top_k=5)
    dlogits = token_logprobs_bwd(logits, targets, r.stats, r.entropy, dlogp)
"""
from __future__ import annotations

import ctypes
from collections import namedtuple
from dataclasses import dataclass

import torch
from torch.autograd.function import once_differentiable

from . import (QN_BF16, QN_EALIGN, QN_F32, NF4State, _Act8, _BlockNorm, _check, _dev,
               _linear_args, _mark_nodes, _opts, _ptr, _refuse_default_stream, _room, _stream,
               _written, load_library)

ACT8_BLOCK = 64
MAX_TOP = 32  # alternatives of a row
GATE_NONE, GATE_CHANNEL, GATE_ROW, GATE_ELEMENT = range(4)
_DTYPES = {torch.bfloat16: QN_BF16, torch.float32: QN_F32}
# Allocations below are written torch.empty(M, cols, ..) or empty_like: 1.2 us of a
# small call's host time each, where torch.empty((M, cols), ..) takes 1.7.


def _aligned(status: int, *ts: torch.Tensor | None):
    """After a call that returned QN_EALIGN: its inputs, those that start between 16-byte
    boundaries (slices of larger tensors) as copies, for a second try; None where that
    is not it.  (Asked beforehand, it is 0.3 to 0.7 us of every small call.)"""
    if status != QN_EALIGN or not any(t is not None and t.data_ptr() % 16 for t in ts):
        return None
    return [t.clone() if t is not None and t.data_ptr() % 16 else t for t in ts]


# ------------------------------------------------- activation checkpoints in 8 bits
@dataclass
class Act8:
    """An activation [M, cols] in 8 bits: int8 codes and one exponent byte E
    for every 64 columns of a row; element = code * 2^(E - 127)."""
    codes: torch.Tensor  # int8 [M, cols]
    exps: torch.Tensor   # uint8 [M, ceil(cols / 64)]

    def nbytes(self) -> int:
        return self.codes.numel() + self.exps.numel()

    def c_struct(self) -> _Act8:
        return _Act8(self.codes.data_ptr(), self.exps.data_ptr())


def _blocks(cols: int) -> int:
    return (cols + ACT8_BLOCK - 1) // ACT8_BLOCK


def _act8(x8: Act8, M: int, cols: int, name: str = "x8") -> Act8:
    if not isinstance(x8, Act8):
        raise ValueError(f"{name} must be an Act8")
    _dev(x8.codes, torch.int8, f"{name}.codes")
    _dev(x8.exps, torch.uint8, f"{name}.exps")
    if x8.codes.shape != (M, cols) or x8.exps.shape != (M, _blocks(cols)):
        raise ValueError(f"{name} must hold codes [{M}, {cols}] and exps [{M}, {_blocks(cols)}]")
    return x8


def _empty_act8(M: int, cols: int, device) -> Act8:
    return Act8(torch.empty(M, cols, dtype=torch.int8, device=device),
                torch.empty(M, _blocks(cols), dtype=torch.uint8, device=device))


def act8_pack(x: torch.Tensor, out: Act8 | None = None) -> Act8:
    """The 8-bit checkpoint of x, bf16 [..., cols] (leading dimensions are
    rows)."""
    x = _dev(x, torch.bfloat16, "x")
    if x.dim() < 1 or x.shape[-1] < 1:
        raise ValueError("x must be [..., cols] with cols >= 1")
    cols = x.shape[-1]
    M = x.numel() // cols
    given = out is not None
    out = _act8(out, M, cols, "out") if given else _empty_act8(M, cols, x.device)
    rc = load_library().act8_pack(x.data_ptr(), M, cols, out.codes.data_ptr(),
                                  out.exps.data_ptr(), _stream(x.device))
    if rc:
        again = _aligned(rc, x)
        return act8_pack(*again, out=out) if again else _check(rc)
    if given:
        _written(out.codes, out.exps)
    return out


def act8_unpack(x8: Act8, out: torch.Tensor | None = None) -> torch.Tensor:
    """The values a checkpoint stands for, bf16 [M, cols] (exact)."""
    if not isinstance(x8, Act8) or x8.codes.dim() != 2:
        raise ValueError("x8 must be an Act8 with codes [M, cols]")
    M, cols = x8.codes.shape
    _act8(x8, M, cols)
    given = out is not None
    if not given:
        out = torch.empty(M, cols, dtype=torch.bfloat16, device=x8.codes.device)
    elif _dev(out, torch.bfloat16, "out").shape != (M, cols):
        raise ValueError(f"out must be [{M}, {cols}]")
    s = x8.c_struct()
    rc = load_library().act8_unpack(ctypes.byref(s), M, cols, out.data_ptr(),
                                    _stream(out.device))
    if rc:
        again = _aligned(rc, x8.codes, x8.exps)
        return act8_unpack(Act8(*again), out=out) if again else _check(rc)
    if given:
        _written(out)
    return out


def qlora_linear_bwd_act8(st: NF4State, x8: Act8, dY: torch.Tensor, A: torch.Tensor,
                          B: torch.Tensor, alpha: float, u: torch.Tensor, need_dx: bool = True,
                          workspace: torch.Tensor | None = None, rslora: bool = False,
                          dropout_mask: torch.Tensor | None = None, dropout_p: float = 0.0,
                          drop=None):
    """qlora_linear_bwd with the forward's input kept as an 8-bit checkpoint
    and u the forward's saved u.  Returns (dX bf16 [M, d_in] or None,
    dA fp32 [r, d_in], dB fp32 [d_out, r])."""
    L = load_library()
    dY = _dev(dY, torch.bfloat16, "dY")
    A = _dev(A, torch.bfloat16, "A")
    B = _dev(B, torch.bfloat16, "B")
    u = _dev(u, torch.float32, "u")
    if not isinstance(x8, Act8) or x8.codes.dim() != 2:
        raise ValueError("x8 must be an Act8 with codes [M, cols]")
    M, r = _linear_args(st, x8.codes, A, B)
    _act8(x8, M, st.cols)
    if dY.shape != (M, st.rows):
        raise ValueError(f"dY must be [{M}, {st.rows}]")
    if u.shape != (M, r):
        raise ValueError(f"u must be [{M}, {r}]")
    dev = dY.device
    dX = torch.empty(M, st.cols, dtype=torch.bfloat16, device=dev) if need_dx else None
    dA = torch.empty(r, st.cols, dtype=torch.float32, device=dev)
    dB = torch.empty(st.rows, r, dtype=torch.float32, device=dev)
    if drop is not None:
        from . import _one_dropout, _qlora_bwd_drop
        _one_dropout(dropout_mask, dropout_p)
        rc = _qlora_bwd_drop(st, None, x8, dY, A, B, r, alpha, rslora, drop, u, dX, dA, dB,
                             workspace)
        if rc:
            again = _aligned(rc, x8.codes, x8.exps, dY, A, B, u)
            if not again:
                _check(rc)
            codes, exps, dY, A, B, u = again
            return qlora_linear_bwd_act8(st, Act8(codes, exps), dY, A, B, alpha, u,
                                         need_dx=need_dx, workspace=workspace, rslora=rslora,
                                         drop=drop)
        return dX, dA, dB
    o = _opts(rslora, dropout_mask, dropout_p, M * st.cols)
    need = L.qlora_linear_bwd_act8_workspace(M, st.rows, st.cols, r, int(need_dx))
    workspace = _room(workspace, need, dev)
    s, c = st.c_struct(), x8.c_struct()
    rc = L.qlora_linear_bwd_act8(ctypes.byref(s), ctypes.byref(c), dY.data_ptr(), M,
                                 A.data_ptr(), B.data_ptr(), r, float(alpha),
                                 ctypes.byref(o) if o is not None else None, u.data_ptr(),
                                 _ptr(dX), dA.data_ptr(), dB.data_ptr(), workspace.data_ptr(),
                                 workspace.numel(), _stream(dev))
    if rc:
        again = _aligned(rc, x8.codes, x8.exps, dY, A, B, u)
        if not again:
            _check(rc)
        codes, exps, dY, A, B, u = again
        return qlora_linear_bwd_act8(st, Act8(codes, exps), dY, A, B, alpha, u, need_dx=need_dx,
                                     workspace=workspace, rslora=rslora,
                                     dropout_mask=dropout_mask, dropout_p=dropout_p)
    return dX, dA, dB


# --------------------------------------------------------------- block norms
BlockNormGrads = namedtuple("BlockNormGrads", "dh do dgate dw_post dw_pre")


def _norm_args(h, w_pre, o, w_post, gate, scale, eps):
    """The C argument struct of a block norm on h [..., D]."""
    if not isinstance(h, torch.Tensor) or h.dtype not in _DTYPES:
        raise ValueError("h must be a bfloat16 or float32 tensor")
    _dev(h, h.dtype, "h")
    if h.dim() < 1 or h.shape[-1] < 1:
        raise ValueError("h must be [..., D] with D >= 1")
    shape, D = h.shape, h.shape[-1]
    M = h.numel() // D
    if not isinstance(w_pre, torch.Tensor) or w_pre.dtype not in _DTYPES:
        raise ValueError("w_pre must be a bfloat16 or float32 tensor")
    wt = w_pre.dtype
    if _dev(w_pre, wt, "w_pre").shape != (D,):
        raise ValueError(f"w_pre must be [{D}]")
    if o is None:
        if w_post is not None or gate is not None:
            raise ValueError("w_post and gate belong to a block output o")
    elif _dev(o, torch.bfloat16, "o").shape != shape:
        raise ValueError("o must have h's shape")
    if w_post is not None and _dev(w_post, wt, "w_post").shape != (D,):
        raise ValueError(f"w_post must be [{D}]")
    kind = GATE_NONE
    if gate is not None:
        gs = gate.shape if isinstance(gate, torch.Tensor) else None
        if gs == (D,):
            kind = GATE_CHANNEL
            _dev(gate, wt, "gate")
        elif gs == shape[:-1] + (1,):
            kind = GATE_ROW
            _dev(gate, torch.bfloat16, "gate")
        elif gs == shape:
            kind = GATE_ELEMENT
            _dev(gate, torch.bfloat16, "gate")
        else:
            raise ValueError(f"gate must be [{D}], [..., 1] or h's shape")
    return _BlockNorm(M, D, w_pre.data_ptr(), _ptr(w_post), _ptr(gate), _DTYPES[h.dtype],
                      _DTYPES[wt], kind, scale, eps)


def block_norm_fwd(h: torch.Tensor, w_pre: torch.Tensor, o: torch.Tensor | None = None,
                   w_post: torch.Tensor | None = None, gate: torch.Tensor | None = None,
                   scale: float = 1.0, eps: float = 1e-6, pack: bool = False):
    """h' = h + scale * gate * post(o) and y = RMSNorm(h') * w_pre on h [..., D]
    (bf16 or fp32); post is RMSNorm(o) * w_post, or o itself without w_post.
    gate: [D] (a channel's), [..., 1] (a row's) or h's shape.  Without o: the
    norm of h alone.  Returns (h' in h's type -- h itself without o --, y bf16,
    y's Act8 with pack or None)."""
    n = _norm_args(h, w_pre, o, w_post, gate, scale, eps)
    dev = h.device
    h_new = None if o is None else torch.empty_like(h)
    y = torch.empty_like(h, dtype=torch.bfloat16)
    x8 = _empty_act8(n.M, n.D, dev) if pack else None
    rc = load_library().block_norm_fwd(
        ctypes.byref(n), h.data_ptr(), _ptr(o), _ptr(h_new), y.data_ptr(),
        x8.codes.data_ptr() if pack else None, x8.exps.data_ptr() if pack else None,
        _stream(dev))
    if rc:
        again = _aligned(rc, h, w_pre, o, w_post, gate)
        if not again:
            _check(rc)
        h_new, y, x8 = block_norm_fwd(*again, scale=scale, eps=eps, pack=pack)
    return (h if o is None else h_new), y, x8


def block_norm_bwd(dy: torch.Tensor, h_new: torch.Tensor, w_pre: torch.Tensor,
                   dh_new: torch.Tensor | None = None, o: torch.Tensor | None = None,
                   w_post: torch.Tensor | None = None, gate: torch.Tensor | None = None,
                   scale: float = 1.0, eps: float = 1e-6, need_weights: bool = True,
                   need_gate: bool = True,
                   workspace: torch.Tensor | None = None) -> BlockNormGrads:
    """Gradients of block_norm_fwd from dy (of y) and dh_new (of h'; None:
    zero), with its h' (h itself without o) and o: dh in h's type, do bf16,
    dgate (fp32 for [D] and [..., 1] gates, bf16 for full ones), dw_post and
    dw_pre fp32 [D] (None without need_weights, for frozen norms)."""
    L = load_library()
    n = _norm_args(h_new, w_pre, o, w_post, gate, scale, eps)
    if _dev(dy, torch.bfloat16, "dy").shape != h_new.shape:
        raise ValueError("dy must have h_new's shape")
    if dh_new is not None and _dev(dh_new, h_new.dtype, "dh_new").shape != h_new.shape:
        raise ValueError("dh_new must have h_new's shape")
    dev, D = h_new.device, n.D
    dh = torch.empty_like(h_new)
    do = None if o is None else torch.empty_like(o)
    dgate = None
    if gate is not None and need_gate:
        dgate = torch.empty_like(gate, dtype=torch.bfloat16
                                 if n.gate_kind == GATE_ELEMENT else torch.float32)
    dw_pre = dw_post = None
    if need_weights:
        dw_pre = torch.empty(D, dtype=torch.float32, device=dev)
        if w_post is not None:
            dw_post = torch.empty(D, dtype=torch.float32, device=dev)
    need = L.block_norm_bwd_workspace(ctypes.byref(n), int(need_weights), int(dgate is not None))
    if need > 0:
        workspace = _room(workspace, need, dev)
    rc = L.block_norm_bwd(ctypes.byref(n), dy.data_ptr(), _ptr(dh_new), h_new.data_ptr(),
                          _ptr(o), dh.data_ptr(), _ptr(do), _ptr(dgate), _ptr(dw_post),
                          _ptr(dw_pre), _ptr(workspace),
                          0 if workspace is None else workspace.numel(), _stream(dev))
    if rc:
        again = _aligned(rc, dy, h_new, w_pre, dh_new, o, w_post, gate)
        return block_norm_bwd(*again, scale=scale, eps=eps, need_weights=need_weights,
                              need_gate=need_gate, workspace=workspace) if again else _check(rc)
    return BlockNormGrads(dh, do, dgate, dw_post, dw_pre)


class _BlockNormFn(torch.autograd.Function):
    @staticmethod
    def forward(ctx, h, o, w_pre, w_post, gate, scale, eps, pack):
        h_new, y, x8 = block_norm_fwd(h, w_pre, o=o, w_post=w_post, gate=gate, scale=scale,
                                      eps=eps, pack=pack)
        ctx.set_materialize_grads(False)
        ctx.save_for_backward(h_new, o, w_pre, w_post, gate)
        ctx.scale, ctx.eps = scale, eps
        codes, exps = (x8.codes, x8.exps) if pack else (None, None)
        if pack:
            ctx.mark_non_differentiable(codes, exps)
        return (None if o is None else h_new), y, codes, exps

    @staticmethod
    @once_differentiable
    def backward(ctx, dh_new, dy, *_):
        _refuse_default_stream(ctx)
        h_new, o, w_pre, w_post, gate = ctx.saved_tensors
        need = ctx.needs_input_grad
        if dy is None:
            if not (need[1] or need[3] or need[4]):  # h' alone, and only h behind it
                return dh_new, None, None, None, None, None, None, None
            dy = torch.zeros(h_new.shape, dtype=torch.bfloat16, device=h_new.device)
        g = block_norm_bwd(dy.contiguous(), h_new, w_pre,
                           dh_new=None if dh_new is None else dh_new.contiguous(), o=o,
                           w_post=w_post, gate=gate, scale=ctx.scale, eps=ctx.eps,
                           need_weights=need[2] or need[3], need_gate=need[4])
        cast = lambda d, w: None if d is None else d.to(w.dtype)  # noqa: E731
        return (g.dh, g.do, cast(g.dw_pre, w_pre), cast(g.dw_post, w_post),
                cast(g.dgate, gate), None, None, None)


class BlockNorm(torch.nn.Module):
    """The end of one block and the start of the next: forward(h, o) gives
    (h', y, Act8 of y or None) as block_norm_fwd does, with gradients; o None:
    the norm of h alone.  post: a norm on the block's output; gate: a learned
    gate for every channel (starts at one); scale: the residual scale."""

    def __init__(self, dim: int, post: bool = False, gate: bool = False, scale: float = 1.0,
                 eps: float = 1e-6, dtype=torch.float32, device="cuda"):
        super().__init__()
        one = lambda on: torch.nn.Parameter(  # noqa: E731
            torch.ones(dim, dtype=dtype, device=device)) if on else None
        self.w_pre, self.w_post, self.gate = one(True), one(post), one(gate)
        self.scale, self.eps = float(scale), float(eps)

    def forward(self, h, o=None, pack=False):
        w_post, gate = (None, None) if o is None else (self.w_post, self.gate)
        h_new, y, codes, exps = _BlockNormFn.apply(h, o, self.w_pre, w_post, gate, self.scale,
                                                   self.eps, pack)
        _mark_nodes(y)
        return (h if o is None else h_new), y, Act8(codes, exps) if pack else None


# ------------------------------------------------------ token log probabilities
TokenLogprobs = namedtuple("TokenLogprobs", "logp entropy stats top_logp top_ids")


def _logits(logits, targets, name="logits"):
    if not isinstance(logits, torch.Tensor) or not logits.is_cuda:
        raise ValueError(f"{name} must be a CUDA (HIP) tensor")
    if logits.dtype not in _DTYPES:
        raise ValueError(f"{name} must be bfloat16 or float32, got {logits.dtype}")
    if logits.dim() != 2 or logits.shape[1] < 1:
        raise ValueError(f"{name} must be [T, V] with V >= 1")
    T, V = logits.shape
    ld = logits.stride(0) if T > 1 else V
    if (V > 1 and logits.stride(1) != 1) or ld < V:
        raise ValueError(f"{name}' rows must be contiguous and must not overlap")
    if targets is not None and _dev(targets, torch.int64, "targets").shape != (T,):
        raise ValueError(f"targets must be [{T}]")
    return T, V, ld


def token_logprobs_fwd(logits: torch.Tensor, targets: torch.Tensor | None = None,
                       scale: float = 1.0, top_k: int = 0,
                       workspace: torch.Tensor | None = None) -> TokenLogprobs:
    """With p = softmax(scale * logits) over each row of logits [T, V] (bf16 or
    fp32; rows may be wider than V apart): logp [T] = ln p of the targets
    (None without targets; 0 where a target is negative), entropy [T], stats
    [T, 2] for the backward, and the top_k most likely tokens of each row
    (top_logp, top_ids int32 [T, top_k], descending, ties to the lower index;
    None with top_k = 0)."""
    L = load_library()
    T, V, ld = _logits(logits, targets)
    if not 0 <= top_k <= min(MAX_TOP, V):
        raise ValueError(f"top_k must be 0 .. {min(MAX_TOP, V)}")
    dev = logits.device
    f32 = torch.float32
    entropy = torch.empty(T, dtype=f32, device=dev)
    logp = None if targets is None else torch.empty_like(entropy)
    stats = torch.empty(T, 2, dtype=f32, device=dev)
    top_logp = top_ids = None
    if top_k:
        top_logp = torch.empty(T, top_k, dtype=f32, device=dev)
        top_ids = torch.empty(T, top_k, dtype=torch.int32, device=dev)
    dt = _DTYPES[logits.dtype]
    need = L.token_logprobs_workspace(T, V, dt, top_k)
    if need > 0:
        workspace = _room(workspace, need, dev)
    _check(L.token_logprobs_fwd(logits.data_ptr(), dt, T, V, ld, _ptr(targets), scale, top_k,
                                _ptr(logp), entropy.data_ptr(), stats.data_ptr(), _ptr(top_logp),
                                _ptr(top_ids), _ptr(workspace),
                                0 if workspace is None else workspace.numel(), _stream(dev)))
    return TokenLogprobs(logp, entropy, stats, top_logp, top_ids)


def token_logprobs_bwd(logits: torch.Tensor, targets: torch.Tensor | None, stats: torch.Tensor,
                       entropy: torch.Tensor | None, dlogp: torch.Tensor | None,
                       dentropy: torch.Tensor | None = None, scale: float = 1.0,
                       out: torch.Tensor | None = None) -> torch.Tensor:
    """The gradient of token_logprobs_fwd with respect to the logits, in their
    type, from dlogp [T] and/or dentropy [T] and the forward's stats and
    entropy.  out may be the logits themselves."""
    L = load_library()
    T, V, ld = _logits(logits, targets)
    if dlogp is None and dentropy is None:
        raise ValueError("dlogp or dentropy is needed")
    if dlogp is not None and targets is None:
        raise ValueError("dlogp needs targets")
    if dentropy is not None and entropy is None:
        raise ValueError("dentropy needs the forward's entropy")
    if _dev(stats, torch.float32, "stats").shape != (T, 2):
        raise ValueError(f"stats must be [{T}, 2]")
    for name, t in (("entropy", entropy), ("dlogp", dlogp), ("dentropy", dentropy)):
        if t is not None and _dev(t, torch.float32, name).shape != (T,):
            raise ValueError(f"{name} must be [{T}]")
    given = out is not None
    if not given:
        out = torch.empty(T, V, dtype=logits.dtype, device=logits.device)
    elif out.dtype != logits.dtype or out.shape != logits.shape:
        raise ValueError("out must have the logits' type and shape")
    _, _, ldd = _logits(out, None, "out")
    rc = L.token_logprobs_bwd(logits.data_ptr(), _DTYPES[logits.dtype], T, V, ld, _ptr(targets),
                              scale, stats.data_ptr(), _ptr(entropy), _ptr(dlogp),
                              _ptr(dentropy), out.data_ptr(), ldd, _stream(logits.device))
    if rc:
        again = _aligned(rc, stats, entropy, dlogp, dentropy)
        return token_logprobs_bwd(logits, targets, *again, scale=scale,
                                  out=out) if again else _check(rc)
    if given:
        _written(out)
    return out


class _TokenLogprobsFn(torch.autograd.Function):
    @staticmethod
    def forward(ctx, logits, targets, scale, top_k):
        r = token_logprobs_fwd(logits, targets, scale=scale, top_k=top_k)
        ctx.set_materialize_grads(False)
        ctx.save_for_backward(logits, targets, r.stats, r.entropy)
        ctx.scale = scale
        ctx.mark_non_differentiable(*[t for t in (r.stats, r.top_logp, r.top_ids)
                                      if t is not None])
        return r.logp, r.entropy, r.stats, r.top_logp, r.top_ids

    @staticmethod
    @once_differentiable
    def backward(ctx, dlogp, dentropy, *_):
        logits, targets, stats, entropy = ctx.saved_tensors
        if dlogp is None and dentropy is None:
            return None, None, None, None
        c = lambda t: None if t is None else t.contiguous()  # noqa: E731
        return token_logprobs_bwd(logits, targets, stats, entropy, c(dlogp), c(dentropy),
                                  scale=ctx.scale), None, None, None


def token_logprobs(logits: torch.Tensor, targets: torch.Tensor | None = None, scale: float = 1.0,
                   top_k: int = 0) -> TokenLogprobs:
    """token_logprobs_fwd with gradients through logp and entropy."""
    return TokenLogprobs(*_TokenLogprobsFn.apply(logits, targets, scale, top_k))
