"""The linear on weights in MXFP4, the matrix cores' own 4-bit format, and
dropout whose mask is drawn from a counter where it is used and never kept.

As in the package's other calls, the functions carry the C names and only check
and marshal arguments; outputs and workspaces are torch allocations on the
current stream.

    w = mx4_quantize(W)                          # W fp32 or bf16 [d_out, d_in]
    drop = Dropout(0.05, seed=7, offset=3)
    y, u = mx4_linear_fwd(w, x, A, B, alpha, drop=drop)
    dX, dA, dB = mx4_linear_bwd(w, x, dY, A, B, alpha, u, drop=drop)
    y, u = qlora_linear_fwd(st, x, A, B, alpha, drop=drop)   # on an NF4 state
    h = dropout(h, drop)                         # an activation by itself
"""
from __future__ import annotations

import ctypes
import functools
from dataclasses import dataclass

import torch
from torch.autograd.function import once_differentiable

from . import (NF4State, QNError, _check, _dev, _Dropout, _MX4, _ptr,  # noqa: F401
               _refuse_default_stream, _room, _stream, load_library)
from .finetune import _DTYPES, Act8, _act8, _aligned, _written

MX4_BLOCK = 32   # columns of a row that share a scale
MX4_STEP = 256   # columns that a row of codes is padded to


@functools.lru_cache(maxsize=None)
def _one_device() -> bool:
    return torch.cuda.device_count() == 1


def _here(*ts: torch.Tensor | None) -> bool:
    """Whether the tensors, which must share a device, lie on the current one (kernels
    are launched there).  (With one device there is nothing to ask: 1.5 us of a small
    call's 12.)"""
    if _one_device():
        return True
    dev = None
    for t in ts:
        if t is not None:
            if dev is not None and t.device != dev:
                raise ValueError("all tensors must be on one device")
            dev = t.device
    return dev is None or dev.index == torch.cuda.current_device()


@functools.lru_cache(maxsize=4096)
def _need(*sizes: int) -> int:
    """mx4_linear_workspace(*sizes) (asked again each time it is 0.8 us)."""
    return load_library().mx4_linear_workspace(*sizes)


@functools.lru_cache(maxsize=4096)
def _need_drop(*sizes: int) -> int:
    return load_library().qlora_linear_drop_workspace(*sizes)


# ------------------------------------------------------- dropout from a counter
@dataclass(frozen=True, eq=False)
class Dropout:
    """Dropout with probability p (taken in steps of 2^-16), its mask a function
    of seed, offset and the element's number: the same key draws the same mask in the
    forward and in the backward, and nothing is kept between them.  offset tells the
    uses of one seed apart (layers, steps).  step: an int64 tensor of one element on
    the device that is added to offset when the kernels run, so that a captured
    graph draws another mask at each replay; it must not change between a forward
    and its backward.  Offset and step are one sum: uses in one graph whose offsets
    lie nearer than step gets have each other's masks at other replays."""
    p: float
    seed: int
    offset: int = 0
    step: torch.Tensor | None = None

    def __post_init__(self):
        if not 0.0 <= self.p < 1.0:
            raise ValueError("p must be in [0, 1)")
        for name in ("seed", "offset"):
            v = getattr(self, name)
            if not isinstance(v, int) or not 0 <= v < 1 << 64:
                raise ValueError(f"{name} must be a whole number below 2^64")
        if self.step is not None and _dev(self.step, torch.int64, "step").numel() != 1:
            raise ValueError("step must hold one int64")

    def c_struct(self) -> _Dropout:
        # (the C side has p in 32 bits, where the nearest number may be 1, which it refuses)
        return _Dropout(self.seed, self.offset, _ptr(self.step), min(self.p, 1 - 2.0 ** -24))


def _drop(drop: Dropout | None, *beside: torch.Tensor):
    """The C argument of drop (a pointer or None)."""
    if drop is None:
        return None
    if not isinstance(drop, Dropout):
        raise ValueError("drop must be a Dropout")
    if drop.step is not None:
        _here(drop.step, *beside)
    return ctypes.byref(drop.c_struct())


def dropout_apply(x: torch.Tensor, drop: Dropout, out: torch.Tensor | None = None) -> torch.Tensor:
    """x (bf16 or fp32, any shape) with the elements that drop drops set to zero and the
    others scaled up; out may be x.  The same call on the gradient is its backward."""
    if not isinstance(x, torch.Tensor) or x.dtype not in _DTYPES:
        raise ValueError("x must be a bfloat16 or float32 tensor")
    _dev(x, x.dtype, "x")
    if not isinstance(drop, Dropout):
        raise ValueError("drop must be a Dropout")
    given = out is not None
    if not given:
        out = torch.empty_like(x)
    elif _dev(out, x.dtype, "out").shape != x.shape:
        raise ValueError("out must have x's shape")
    if given:
        a, b, n = x.data_ptr(), out.data_ptr(), x.numel() * x.element_size()
        if a != b and a < b + n and b < a + n:
            raise ValueError("out may be x itself but may not overlap it otherwise")
    if not _here(x, out):
        with torch.cuda.device(x.device):
            return dropout_apply(x, drop, out)
    _check(load_library().dropout_apply(x.data_ptr(), _DTYPES[x.dtype], x.numel(),
                                        _drop(drop, x), out.data_ptr(), _stream(x.device)))
    if given:
        _written(out)
    return out


class _DropoutFn(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, drop):
        ctx.save_for_backward(drop.step)  # (a step changed before the backward is an error)
        ctx.drop = drop
        return dropout_apply(x, drop)

    @staticmethod
    @once_differentiable
    def backward(ctx, dy):
        ctx.saved_tensors
        return dropout_apply(dy.contiguous(), ctx.drop), None


def dropout(x: torch.Tensor, drop: Dropout | None) -> torch.Tensor:
    """dropout_apply with gradients; x itself without drop."""
    return x if drop is None else _DropoutFn.apply(x, drop)


# ---------------------------------------------------------------------- MXFP4
@dataclass
class MX4:
    """A matrix [rows, cols] in MXFP4 (layout in the header): E2M1 codes, two a
    byte, rows padded to 256 columns, and a power-of-two scale for every 32 columns
    of a row, in the order in which the matrix instructions take them."""
    codes: torch.Tensor   # uint8 [rows, 128 J], J = ceil(cols / 256)
    scales: torch.Tensor  # uint8 [ceil(rows / 32), J, 256]
    rows: int
    cols: int

    def c_struct(self) -> _MX4:
        return _MX4(self.codes.data_ptr(), self.scales.data_ptr(), self.rows, self.cols)

    @property
    def device(self):
        return self.codes.device

    def nbytes(self) -> int:
        return self.codes.numel() + self.scales.numel()


def _shapes(rows: int, cols: int):
    J = (cols + MX4_STEP - 1) // MX4_STEP
    return (rows, 128 * J), ((rows + 31) // 32, J, 256)


def _mx4(w: MX4, name: str = "w") -> MX4:
    if not isinstance(w, MX4):
        raise ValueError(f"{name} must be an MX4")
    codes, scales = _shapes(w.rows, w.cols)
    if _dev(w.codes, torch.uint8, "codes").shape != codes:
        raise ValueError(f"{name}.codes must be {list(codes)}")
    if _dev(w.scales, torch.uint8, "scales").shape != scales:
        raise ValueError(f"{name}.scales must be {list(scales)}")
    return w


def mx4_quantize(x: torch.Tensor, out: MX4 | None = None) -> MX4:
    """x [..., cols], bf16 or fp32, in MXFP4 (leading dimensions are rows)."""
    if not isinstance(x, torch.Tensor) or x.dtype not in _DTYPES:
        raise ValueError("x must be a bfloat16 or float32 tensor")
    _dev(x, x.dtype, "x")
    if x.dim() < 1 or x.shape[-1] < 1:
        raise ValueError("x must be [..., cols] with cols >= 1")
    cols = x.shape[-1]
    rows = x.numel() // cols
    given = out is not None
    if not given:
        codes, scales = _shapes(rows, cols)
        out = MX4(torch.empty(*codes, dtype=torch.uint8, device=x.device),
                  torch.empty(*scales, dtype=torch.uint8, device=x.device), rows, cols)
    elif (_mx4(out, "out").rows, out.cols) != (rows, cols):
        raise ValueError(f"out must be [{rows}, {cols}]")
    if not _here(x, out.codes, out.scales):
        with torch.cuda.device(x.device):
            return mx4_quantize(x, out)
    rc = load_library().mx4_quantize(x.data_ptr(), _DTYPES[x.dtype], rows, cols,
                                     out.codes.data_ptr(), out.scales.data_ptr(),
                                     _stream(x.device))
    if rc:
        again = _aligned(rc, x)
        return mx4_quantize(*again, out=out) if again else _check(rc)
    if given:
        _written(out.codes, out.scales)
    return out


def mx4_dequantize(w: MX4, dtype=torch.bfloat16, out: torch.Tensor | None = None) -> torch.Tensor:
    """The values w stands for, [rows, cols] in bf16 or fp32 (exact in both)."""
    _mx4(w)
    if dtype not in _DTYPES:
        raise ValueError("dtype must be bfloat16 or float32")
    given = out is not None
    if not given:
        out = torch.empty(w.rows, w.cols, dtype=dtype, device=w.device)
    elif _dev(out, dtype, "out").shape != (w.rows, w.cols):
        raise ValueError(f"out must be [{w.rows}, {w.cols}]")
    if not _here(w.codes, w.scales, out):
        with torch.cuda.device(w.device):
            return mx4_dequantize(w, dtype, out)
    _check(load_library().mx4_dequantize(ctypes.byref(w.c_struct()), _DTYPES[dtype],
                                         out.data_ptr(), _stream(w.device)))
    if given:
        _written(out)
    return out


def _adapter(w, M, A, B, drop):
    """The rank of an adapter beside w (0: none)."""
    if A is None and B is None:
        if drop is not None:
            raise ValueError("drop belongs to an adapter")
        return 0
    if A is None or B is None:
        raise ValueError("A and B come together")
    _dev(A, torch.bfloat16, "A")
    _dev(B, torch.bfloat16, "B")
    r = A.shape[0]
    if A.dim() != 2 or A.shape[1] != w.cols or B.shape != (w.rows, r):
        raise ValueError(f"A must be [r, {w.cols}] and B [{w.rows}, r]")
    return r


def _workspace(need: int, given: torch.Tensor | None, device) -> torch.Tensor:
    ws = _room(given, need, device)
    if ws.dtype != torch.uint8:
        raise ValueError("workspace must be a uint8 tensor")
    return ws


def mx4_linear_fwd(w: MX4, x: torch.Tensor, A: torch.Tensor | None = None,
                   B: torch.Tensor | None = None, alpha: float = 0.0, save_u: bool = True,
                   y: torch.Tensor | None = None, workspace: torch.Tensor | None = None,
                   rslora: bool = False, drop: Dropout | None = None):
    """y = Q(x) W^T + s u B^T with u = drop(x) A^T and Q the rounding of x [M, cols]
    (bf16) to MXFP4; s as in qlora_linear_fwd.  Without A and B: the product
    alone, of any sizes.  Returns (y bf16 [M, rows], u fp32 [M, r] or None)."""
    _mx4(w)
    if _dev(x, torch.bfloat16, "x").dim() != 2 or x.shape[1] != w.cols:
        raise ValueError(f"x must be [M, {w.cols}]")
    M = x.shape[0]
    r = _adapter(w, M, A, B, drop)
    given = y is not None
    if not given:
        y = torch.empty(M, w.rows, dtype=torch.bfloat16, device=x.device)
    elif _dev(y, torch.bfloat16, "y").shape != (M, w.rows):
        raise ValueError(f"y must be [{M}, {w.rows}]")
    if not _here(w.codes, w.scales, x, A, B, y):
        with torch.cuda.device(x.device):
            return mx4_linear_fwd(w, x, A, B, alpha, save_u, y, workspace, rslora, drop)
    L = load_library()
    u = torch.empty(M, r, dtype=torch.float32, device=x.device) if save_u and r else None
    ws = _workspace(_need(M, w.rows, w.cols, r, 0, 0, 0), workspace, x.device)
    rc = L.mx4_linear_fwd(ctypes.byref(w.c_struct()), x.data_ptr(), M, _ptr(A), _ptr(B), r,
                          float(alpha), int(bool(rslora)), _drop(drop, x), y.data_ptr(), _ptr(u),
                          ws.data_ptr(), ws.numel(), _stream(x.device))
    if rc:
        again = _aligned(rc, x, A, B)
        if not again:
            _check(rc)
        return mx4_linear_fwd(w, *again, alpha, save_u, y, workspace, rslora, drop)
    if given:
        _written(y)
    return y, u


def _saved_x(x, M, cols):
    """The forward's input as (bf16 tensor or None, Act8 or None)."""
    if isinstance(x, Act8):
        return None, _act8(x, M, cols, "x")
    if _dev(x, torch.bfloat16, "x").shape != (M, cols):
        raise ValueError(f"x must be [{M}, {cols}] or its Act8")
    return x, None


def mx4_linear_bwd(w: MX4, x, dY: torch.Tensor, A: torch.Tensor | None = None,
                   B: torch.Tensor | None = None, alpha: float = 0.0,
                   u: torch.Tensor | None = None, need_dx: bool = True,
                   workspace: torch.Tensor | None = None, rslora: bool = False,
                   drop: Dropout | None = None):
    """The gradients of mx4_linear_fwd (that of Q taken as each element's own) from
    the forward's x, bf16 or an Act8 of it (then u is needed), and u: (dX bf16
    [M, cols] or None, dA fp32 [r, cols], dB fp32 [rows, r]).  Without A and B: dX
    alone (x unused), the others None."""
    _mx4(w)
    if _dev(dY, torch.bfloat16, "dY").dim() != 2 or dY.shape[1] != w.rows:
        raise ValueError(f"dY must be [M, {w.rows}]")
    M = dY.shape[0]
    r = _adapter(w, M, A, B, drop)
    if not r:
        if not need_dx:
            return None, None, None
        xb = x8 = None
    else:
        xb, x8 = _saved_x(x, M, w.cols)
        if x8 is not None and u is None:
            raise ValueError("u is needed with an Act8")
        if u is not None and _dev(u, torch.float32, "u").shape != (M, r):
            raise ValueError(f"u must be [{M}, {r}]")
    dev = dY.device
    codes, exps = (None, None) if x8 is None else (x8.codes, x8.exps)
    if not _here(w.codes, w.scales, dY, xb, codes, exps, A, B, u):
        with torch.cuda.device(dev):
            return mx4_linear_bwd(w, x, dY, A, B, alpha, u, need_dx, workspace, rslora, drop)
    L = load_library()
    dX = torch.empty(M, w.cols, dtype=torch.bfloat16, device=dev) if need_dx else None
    dA = torch.empty(r, w.cols, dtype=torch.float32, device=dev) if r else None
    dB = torch.empty(w.rows, r, dtype=torch.float32, device=dev) if r else None
    ws = _workspace(_need(M, w.rows, w.cols, r, 1, int(x8 is not None), int(drop is not None)),
                    workspace, dev)
    c8 = ctypes.byref(x8.c_struct()) if x8 is not None else None
    rc = L.mx4_linear_bwd(ctypes.byref(w.c_struct()), _ptr(xb), c8, dY.data_ptr(), M, _ptr(A),
                          _ptr(B), r, float(alpha), int(bool(rslora)), _drop(drop, dY), _ptr(u),
                          _ptr(dX), _ptr(dA), _ptr(dB), ws.data_ptr(), ws.numel(), _stream(dev))
    if rc:
        again = _aligned(rc, xb, codes, exps, dY, A, B, u)
        if not again:
            _check(rc)
        xb, codes, exps, dY, A, B, u = again
        return mx4_linear_bwd(w, xb if x8 is None else Act8(codes, exps), dY, A, B, alpha, u,
                              need_dx, workspace, rslora, drop)
    return dX, dA, dB


# ------------------------------------------------- the NF4 linear under a Dropout
def _qlora_fwd_drop(st: NF4State, x, A, B, r, alpha, rslora, drop, y, u, workspace):
    if not _here(x, A, B, y, st.packed):
        with torch.cuda.device(x.device):
            return _qlora_fwd_drop(st, x, A, B, r, alpha, rslora, drop, y, u, workspace)
    L = load_library()
    M = x.shape[0]
    need = _need_drop(M, st.rows, st.cols, r, 0, 0)
    workspace = _room(workspace, need, x.device)  # (nothing to clear, whatever the route)
    _check(L.qlora_linear_fwd_drop(ctypes.byref(st.c_struct()), x.data_ptr(), M, A.data_ptr(),
                                   B.data_ptr(), r, float(alpha), int(bool(rslora)),
                                   _drop(drop, x), y.data_ptr(), _ptr(u), workspace.data_ptr(),
                                   workspace.numel(), _stream(x.device)))
    return y, u


def _qlora_bwd_drop(st: NF4State, x, x8, dY, A, B, r, alpha, rslora, drop, u, dX, dA, dB,
                    workspace):
    codes, exps = (None, None) if x8 is None else (x8.codes, x8.exps)
    if not _here(dY, x, codes, exps, A, B, u, st.packed):
        with torch.cuda.device(dY.device):
            return _qlora_bwd_drop(st, x, x8, dY, A, B, r, alpha, rslora, drop, u, dX, dA, dB,
                                   workspace)
    L = load_library()
    M = dY.shape[0]
    need = _need_drop(M, st.rows, st.cols, r, 1, int(x8 is not None))
    workspace = _room(workspace, need, dY.device)
    return L.qlora_linear_bwd_drop(
        ctypes.byref(st.c_struct()), _ptr(x), None if x8 is None else ctypes.byref(x8.c_struct()),
        dY.data_ptr(), M, A.data_ptr(), B.data_ptr(), r, float(alpha), int(bool(rslora)),
        _drop(drop, dY), _ptr(u), _ptr(dX), dA.data_ptr(), dB.data_ptr(), workspace.data_ptr(),
        workspace.numel(), _stream(dY.device))


def linear_fwd(w, x, A, B, alpha, rslora=False, drop=None):
    """(y, u) of the linear on either kind of base weight."""
    if isinstance(w, MX4):
        return mx4_linear_fwd(w, x, A, B, alpha, rslora=rslora, drop=drop)
    from . import qlora_linear_fwd
    return qlora_linear_fwd(w, x, A, B, alpha, rslora=rslora, drop=drop)


def linear_bwd(w, x, dY, A, B, alpha, u, need_dx=True, rslora=False, drop=None):
    """(dX, dA, dB) of the linear on either kind of base weight, from x or its Act8."""
    if isinstance(w, MX4):
        return mx4_linear_bwd(w, x, dY, A, B, alpha, u, need_dx=need_dx, rslora=rslora, drop=drop)
    from . import qlora_linear_bwd, qlora_linear_bwd_act8
    f = qlora_linear_bwd_act8 if isinstance(x, Act8) else qlora_linear_bwd
    return f(w, x, dY, A, B, alpha, u, need_dx=need_dx, rslora=rslora, drop=drop)


class _LinearFn(torch.autograd.Function):
    """The adapter linear on either base weight under a Dropout; keep8: what the
    backward needs of x is kept in 8 bits (x8, or x packed here)."""

    @staticmethod
    def forward(ctx, x, A, B, w, alpha, rslora, drop, keep8, x8):
        if x8 is not None:
            _act8(x8, *x.shape)
        y, u = linear_fwd(w, x, A, B, alpha, rslora, drop)
        if keep8 and x8 is None:
            from .finetune import act8_pack
            x8 = act8_pack(x)
        kept = (x8.codes, x8.exps) if keep8 else (x, None)
        # (the step with them: changed before the backward it is an error)
        ctx.save_for_backward(*kept, A, B, u, None if drop is None else drop.step)
        ctx.w, ctx.alpha, ctx.rslora, ctx.drop, ctx.keep8 = w, alpha, rslora, drop, keep8
        return y

    @staticmethod
    @once_differentiable
    def backward(ctx, dY):
        _refuse_default_stream(ctx)
        x, exps, A, B, u, _ = ctx.saved_tensors
        dX, dA, dB = linear_bwd(ctx.w, Act8(x, exps) if ctx.keep8 else x, dY.contiguous(), A, B,
                                ctx.alpha, u, need_dx=ctx.needs_input_grad[0],
                                rslora=ctx.rslora, drop=ctx.drop)
        return dX, dA.to(A.dtype), dB.to(B.dtype), None, None, None, None, None, None
