"""The library's training operators as differentiable torch functions: the
embedding lookup, dropout, linear layers whose operands are quantised to
MXFP4, the root-mean-square norm, and linear layers and gated blocks in 16 bits
whose activations can be kept in 8 (include/zero.h, "training operators").

Buffer management and autograd wiring only; every computation is a call of
the binding on the current stream.  Outputs and workspaces come from torch's
allocator.  A model's parameters are the optimizer's (ZeroAdam's views of
its flat buffer, say); the gradients that backward() leaves in `.grad` go into
a rank's gradient buffer, or `embed_grad` and `Mx4Linear.weight_grad` write them
there directly.  The lookup and dropout can be differentiated any number of
times, everything else once: an attempt at more raises.

Forward and backward can be captured in a CUDA graph.  As with any torch function, no
eager graph of the same leaves may still be alive then (an output that was not
freed, say): torch remembers its stream for the leaves and would draw that stream into the
capture, which fails inside torch's engine.

A product whose waits on the device run out stores nothing, and its call
has long returned: where a program reads its losses it also asks for the counts
(`zero_mx4_timeouts()` for the 4-bit ones, `zero_matmul_timeouts()` for the others, 0 when all is
well), which wait for the device.

    h = embed(table, tokens, pad=0)
    h = dropout(h, 0.1, seed, offset)
    y = layer(h)                     # layer = Mx4Linear(weight)
    h = dropout(y, 0.1, seed, offset + 1, residual=h)
    ...
    opt.step(); layer.refresh()      # the weight changed: quantise it again

and a block in 16 bits, what its backward pass needs kept in 8:

    y, h = rms_norm(x, norm_weight, residual=h)          # h: the sum, the next residual
    y = gated(y, w_gate, w_up, keep8=True)
    h = linear(y, w_down, residual=h, keep8=True)
"""
from __future__ import annotations

import math

import torch
from torch.autograd.graph import increment_version

from . import binding as z

_DT = {torch.float32: z.ZERO_F32, torch.bfloat16: z.ZERO_BF16, torch.float16: z.ZERO_F16}


def _rows_apart(x: torch.Tensor) -> bool:
    """Whether x's rows are runs of consecutive elements that do not overlap."""
    return not (x.shape[1] > 1 and x.stride(1) != 1 or
                x.shape[0] > 1 and x.stride(0) < x.shape[1])


def _gradient(dy: torch.Tensor) -> torch.Tensor:
    """An output's gradient as the library can take it.  torch hands on what the
    next operation's gradient looks like: expanded over the rows after a sum
    over them, say."""
    return dy if _rows_apart(dy) else dy.contiguous()


def _matrix(name: str, x: torch.Tensor) -> torch.Tensor:
    """x itself if the library can take it as rows of elements."""
    if not isinstance(x, torch.Tensor) or not x.is_cuda:
        raise ValueError("%s must be a CUDA tensor" % name)
    if x.dtype not in _DT:
        raise ValueError("%s must be fp32, bf16 or fp16, not %s" % (name, x.dtype))
    if x.dim() != 2:
        raise ValueError("%s must have two dimensions, not %d" % (name, x.dim()))
    if not _rows_apart(x):
        raise ValueError("%s must have consecutive elements in its rows" % name)
    return x


def _stride(x: torch.Tensor) -> int:
    return max(x.stride(0), x.shape[1]) if x.shape[0] > 1 else x.shape[1]


def _tokens(tokens: torch.Tensor, device) -> torch.Tensor:
    if not isinstance(tokens, torch.Tensor) or tokens.dtype not in (torch.int32, torch.int64):
        raise ValueError("tokens must be an int32 or int64 tensor")
    if tokens.device != device:
        raise ValueError("tokens must be on %s" % device)
    return tokens.contiguous()


def _written(*tensors) -> None:
    """The caller's tensors were written, through their addresses: torch's autograd counts
    that as for its own operations in place, so that a backward pass which still needs
    what was there raises instead of using what is there now."""
    increment_version([t for t in tensors if t is not None])


def _same(name: str, x: torch.Tensor, like: torch.Tensor) -> None:
    if x.device != like.device or x.dtype != like.dtype or x.shape != like.shape:
        raise ValueError("%s must match in device, dtype and shape" % name)


# ----------------------------------------------------------------- embedding

def embed_grad(dy: torch.Tensor, tokens: torch.Tensor, grad: torch.Tensor, scale: float = 1.0,
               pad: int = -1, accumulate: bool = False) -> torch.Tensor:
    """The table's gradient from dy (a row a token) into `grad` (a row a table
    row: a view of a rank's gradient buffer, say); accumulate adds to it."""
    _matrix("dy", dy)
    _matrix("grad", grad)
    tokens = _tokens(tokens, grad.device)
    if dy.device != grad.device or dy.shape[1] != grad.shape[1] or dy.shape[0] != tokens.numel():
        raise ValueError("dy must have a row of grad's width for every token, on its device")
    rows, dim = grad.shape
    n = tokens.numel()
    with torch.cuda.device(grad.device):
        need = z.zero_embed_grad_workspace(rows, dim, n)
        ws = torch.empty(need, dtype=torch.uint8, device=grad.device)
        z.zero_embed_grad(dy, _DT[dy.dtype], _stride(dy), tokens, tokens.element_size(), n, pad,
                          scale, grad, _DT[grad.dtype], rows, dim, _stride(grad), accumulate, ws,
                          need)
    _written(grad)
    return grad


class _Embed(torch.autograd.Function):
    @staticmethod
    def forward(ctx, table, tokens, scale, pad, bad):
        flat = _tokens(tokens, table.device).reshape(-1)
        out = torch.empty(flat.numel(), table.shape[1], dtype=table.dtype, device=table.device)
        with torch.cuda.device(table.device):
            z.zero_embed(table, _DT[table.dtype], table.shape[0], table.shape[1], _stride(table),
                         flat, flat.element_size(), flat.numel(), pad, scale, out, table.shape[1],
                         bad)
        ctx.save_for_backward(flat)
        ctx.like, ctx.scale, ctx.pad = table, scale, pad
        return out.view(*tokens.shape, table.shape[1])

    @staticmethod
    def backward(ctx, dy):
        (flat,) = ctx.saved_tensors
        dy = dy.reshape(flat.numel(), ctx.like.shape[1])
        grad = (_EmbedGrad.apply if torch.is_grad_enabled() else _table_grad)(
            dy, flat, ctx.like, ctx.scale, ctx.pad)
        return grad, None, None, None, None


def _table_grad(dy, flat, like, scale, pad):
    grad = torch.empty(like.shape, dtype=like.dtype, device=like.device)
    return embed_grad(_gradient(dy), flat, grad, scale, pad)


class _EmbedGrad(torch.autograd.Function):
    """The lookup's transpose; its own gradient is the lookup again."""
    @staticmethod
    def forward(ctx, dy, flat, like, scale, pad):
        ctx.save_for_backward(flat)
        ctx.scale, ctx.pad = scale, pad
        return _table_grad(dy, flat, like, scale, pad)

    @staticmethod
    def backward(ctx, g):
        (flat,) = ctx.saved_tensors
        return _Embed.apply(_gradient(g), flat, ctx.scale, ctx.pad, None), None, None, None, None


def embed(table: torch.Tensor, tokens: torch.Tensor, scale: float = 1.0, pad: int = -1,
          bad: torch.Tensor | None = None) -> torch.Tensor:
    """scale * table[tokens], rows of zeros for the token `pad` and for ids
    outside the table; those are counted in `bad` (one int64 on the device)."""
    _matrix("table", table)
    if bad is not None and (bad.dtype != torch.int64 or bad.device != table.device):
        raise ValueError("bad must be an int64 tensor on the table's device")
    return _Embed.apply(table, tokens, float(scale), int(pad), bad)


# ------------------------------------------------------------------- dropout

def _drop(x, residual, p, seed, offset):
    x = x.contiguous()
    out = torch.empty_like(x)
    with torch.cuda.device(x.device):
        z.zero_dropout(x, residual, out, _DT[x.dtype], x.numel(), p, seed, offset)
    return out


class _Dropout(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, residual, p, seed, offset):
        ctx.args = p, seed, offset
        return _drop(x, residual, p, seed, offset)

    @staticmethod
    def backward(ctx, dy):
        dx = None
        if ctx.needs_input_grad[0]:
            # the same map of dy; where a graph of it is wanted, differentiable again
            dx = (_Dropout.apply if torch.is_grad_enabled() else _drop)(dy, None, *ctx.args)
        return dx, dy if ctx.needs_input_grad[1] else None, None, None, None


def dropout(x: torch.Tensor, p: float, seed: int, offset: int,
            residual: torch.Tensor | None = None) -> torch.Tensor:
    """residual + x with elements dropped by probability p and the others
    divided by 1 - p.  (seed, offset) names the stream of random words: give
    every call of a step an offset of its own.  The mask is made again in the
    backward pass, not stored."""
    if not isinstance(x, torch.Tensor) or not x.is_cuda or x.dtype not in _DT:
        raise ValueError("x must be an fp32, bf16 or fp16 CUDA tensor")
    if not 0.0 <= p <= 1.0:
        raise ValueError("p must be in [0, 1]")
    if residual is not None:
        _same("residual", residual, x)
        residual = residual.contiguous()
    return _Dropout.apply(x, residual, float(p), int(seed) & (2 ** 64 - 1),
                          int(offset) & (2 ** 64 - 1))


# -------------------------------------------------------------- 4-bit products

class Mx4Matrix:
    """A matrix quantised to MXFP4, blocks along its rows."""

    def __init__(self, rows: int, cols: int, device):
        self.rows, self.cols = rows, cols
        self.q = torch.empty(z.zero_mx4_bytes(rows, cols), dtype=torch.uint8, device=device)

    def values(self, dtype: torch.dtype = torch.float32) -> torch.Tensor:
        out = torch.empty(self.rows, self.cols, dtype=dtype, device=self.q.device)
        with torch.cuda.device(out.device):
            z.zero_mx4_dequantize(self.q, self.rows, self.cols, out, _DT[dtype], self.cols)
        return out


def mx4_quantize(x: torch.Tensor, rows: bool = True, cols: bool = True):
    """(x quantised along its rows, its transpose quantised along x's columns),
    either None where not asked for."""
    _matrix("x", x)
    R, C = x.shape
    q = Mx4Matrix(R, C, x.device) if rows else None
    qt = Mx4Matrix(C, R, x.device) if cols else None
    if not (rows or cols):
        return q, qt
    with torch.cuda.device(x.device):
        z.zero_mx4_quantize(x, _DT[x.dtype], R, C, _stride(x), q.q if q else None,
                            qt.q if qt else None)
    return q, qt


def mx4_matmul(a: Mx4Matrix, b: Mx4Matrix, dtype: torch.dtype = torch.bfloat16,
               out: torch.Tensor | None = None, alpha: float = 1.0,
               accumulate: bool = False) -> torch.Tensor:
    """alpha * A B^T, into (or added to) `out` if that is given."""
    if a.cols != b.cols or a.q.device != b.q.device:
        raise ValueError("the matrices must have as many columns and one device")
    if out is None:
        if accumulate:
            raise ValueError("there is nothing to add to")
        out = torch.empty(a.rows, b.rows, dtype=dtype, device=a.q.device)
    _matrix("out", out)
    if out.shape != (a.rows, b.rows) or out.device != a.q.device:
        raise ValueError("out must be %d by %d on %s" % (a.rows, b.rows, a.q.device))
    with torch.cuda.device(out.device):
        z.zero_mx4_matmul(a.q, a.rows, b.q, b.rows, a.cols, alpha, accumulate, out,
                          _DT[out.dtype], _stride(out))
    _written(out)
    return out


class _Once(torch.autograd.Function):
    """A gradient that depends on what `links` do and cannot be differentiated.
    (torch's once_differentiable does not tie it to them: a derivative with
    respect to given inputs would leave it out and say nothing.)"""
    @staticmethod
    def forward(ctx, grad, *links):
        return grad.clone()

    @staticmethod
    def backward(ctx, g):
        raise RuntimeError("Mx4Linear can be differentiated once: its gradients have none")


class _Linear(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, weight, layer, grads):
        ctx.set_materialize_grads(False)
        ctx.layer, ctx.dtype = layer, x.dtype
        # needs_input_grad tells what the tensors ask for, not whether a
        # backward pass can follow (and here, inside, gradients are always off)
        q, ctx.xt = mx4_quantize(x, True, grads and ctx.needs_input_grad[1])
        # the weight as it was quantised for this forward pass
        ctx.wt = layer.wt if ctx.needs_input_grad[0] else None
        link = None
        if grads:                        # leads back to x and the weight, and holds neither
            link = x.new_empty(0)
            ctx.save_for_backward(link)
        return mx4_matmul(q, layer.w, x.dtype), link

    @staticmethod
    def backward(ctx, dy, _):
        dx = dw = None
        if dy is not None:
            q, qt = mx4_quantize(_gradient(dy), ctx.needs_input_grad[0], ctx.needs_input_grad[1])
            if q is not None:
                dx = mx4_matmul(q, ctx.wt, ctx.dtype)
            if qt is not None:
                dw = mx4_matmul(qt, ctx.xt, ctx.layer.weight.dtype)
            if torch.is_grad_enabled():      # a graph of the gradients is wanted
                (link,) = ctx.saved_tensors
                dx, dw = (None if g is None else _Once.apply(g, dy, link) for g in (dx, dw))
        return dx, dw, None, None


class Mx4Linear:
    """y = x W^T with x, W and, in the backward pass, dy quantised to MXFP4 and
    the products summed in fp32.  The gradients are those of the product of
    the quantised operands, passed straight through the quantisation.

    weight: [n, k]; quantised here, along both of its dimensions, and again by
    refresh(), which belongs after every change of it (an optimizer step)."""

    def __init__(self, weight: torch.Tensor):
        self.weight = weight
        self.w = self.wt = None
        self.refresh()

    def refresh(self) -> None:
        with torch.no_grad():
            self.w, self.wt = mx4_quantize(self.weight.detach())

    def __call__(self, x: torch.Tensor) -> torch.Tensor:
        n, k = self.weight.shape
        if x.dim() < 1 or x.shape[-1] != k or x.device != self.weight.device:
            raise ValueError("x must have rows of %d elements on %s" % (k, self.weight.device))
        rows = x.reshape(-1, k)
        _matrix("x", rows)
        return _Linear.apply(rows, self.weight, self, torch.is_grad_enabled())[0].view(
            *x.shape[:-1], n)

    def weight_grad(self, x: torch.Tensor, dy: torch.Tensor, grad: torch.Tensor,
                    accumulate: bool = False) -> torch.Tensor:
        """The weight's gradient from the layer's input and its output's
        gradient, into `grad` ([n, k]: a view of a rank's gradient buffer)."""
        _, xt = mx4_quantize(x, False, True)
        _, dyt = mx4_quantize(dy, False, True)
        return mx4_matmul(dyt, xt, out=grad, accumulate=accumulate)


# ------------------------------------------------------------- rows in 8 bits

class Packed8:
    """A matrix whose rows are kept in 8 bits with a scale for every 32 elements."""

    def __init__(self, rows: int, cols: int, device):
        self.rows, self.cols = rows, cols
        self.q = torch.empty(z.zero_pack8_bytes(rows, cols), dtype=torch.uint8, device=device)

    def values(self, dtype: torch.dtype = torch.float32) -> torch.Tensor:
        out = torch.empty(self.rows, self.cols, dtype=dtype, device=self.q.device)
        with torch.cuda.device(out.device):
            z.zero_unpack8(self.q, self.rows, self.cols, out, _DT[dtype], self.cols)
        return out


def pack8(x: torch.Tensor) -> Packed8:
    """x (two dimensions) in 8 bits."""
    _matrix("x", x)
    p = Packed8(*x.shape, x.device)
    with torch.cuda.device(x.device):
        z.zero_pack8(x, _DT[x.dtype], *x.shape, _stride(x), p.q)
    return p


def _unpacked(q: torch.Tensor, rows: int, cols: int, dtype: torch.dtype) -> torch.Tensor:
    out = torch.empty(rows, cols, dtype=dtype, device=q.device)
    z.zero_unpack8(q, rows, cols, out, _DT[dtype], cols)
    return out


class _Last(torch.autograd.Function):
    """A gradient that depends on what `links` do and cannot be differentiated;
    `name` says whose."""
    @staticmethod
    def forward(ctx, name, grad, *links):
        ctx.name = name
        return grad.clone()

    @staticmethod
    def backward(ctx, g):
        raise RuntimeError("%s can be differentiated once: its gradients have none" % ctx.name)


def _last(name, grads, *links):
    """The gradients as they are, or, where a graph of them is wanted, tied to
    what they depend on."""
    if not torch.is_grad_enabled():
        return grads
    links = [t for t in links if t is not None]
    return [None if g is None else _Last.apply(name, g, *links) for g in grads]


def _rows(x: torch.Tensor, k: int) -> torch.Tensor:
    """x's rows of k elements as a matrix that the library can take."""
    rows = x.reshape(math.prod(x.shape[:-1]), k)
    return rows if _rows_apart(rows) else rows.contiguous()


# -------------------------------------------------------------------- the norm

class _Norm(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, residual, weight, eps, packed, grads):
        ctx.set_materialize_grads(False)
        rows, dim = x.shape
        y = torch.empty_like(x, memory_format=torch.contiguous_format)
        total = None if residual is None else torch.empty_like(y)
        rstd = torch.empty(rows, dtype=torch.float32, device=x.device) if grads else None
        with torch.cuda.device(x.device):
            z.zero_rms_norm(x, _stride(x), residual,
                            0 if residual is None else _stride(residual), weight, _DT[x.dtype],
                            rows, dim, eps, total, dim, y, dim, packed.q if packed else None,
                            rstd)
        link = None
        if grads:
            link = x.new_empty(0)
            ctx.save_for_backward(x if total is None else total, weight, rstd, link)
            if total is not None and not any(ctx.needs_input_grad[:2]):
                ctx.mark_non_differentiable(total)       # the weight has no part in it
        return y, total, link

    @staticmethod
    def backward(ctx, dy, dtotal, _):
        if dy is None and dtotal is None:
            return (None,) * 6
        total, weight, rstd, link = ctx.saved_tensors
        rows, dim = total.shape
        dx = dw = None
        if dy is None:                       # the norm itself led nowhere
            dx = dtotal
            if ctx.needs_input_grad[2]:
                dw = torch.zeros_like(weight)
        else:
            dy = _gradient(dy)
            dtotal = None if dtotal is None else _gradient(dtotal)
            dx = torch.empty(rows, dim, dtype=total.dtype, device=total.device)
            if ctx.needs_input_grad[2]:
                dw = torch.empty_like(weight)
            with torch.cuda.device(total.device):
                need = z.zero_rms_norm_grad_workspace(rows, dim) if dw is not None else 0
                ws = torch.empty(need, dtype=torch.uint8, device=total.device) if need else None
                dt = _DT[total.dtype]
                z.zero_rms_norm_grad(dy, _stride(dy), dtotal,
                                     0 if dtotal is None else _stride(dtotal), total,
                                     _stride(total), weight, rstd, dt, rows, dim, dx, dim, dw, dt,
                                     False, ws, need)
            dx, dw = _last("rms_norm", (dx, dw), dy, dtotal, link)
        return (dx if ctx.needs_input_grad[0] else None,
                dx if ctx.needs_input_grad[1] else None, dw, None, None, None)


def rms_norm(x: torch.Tensor, weight: torch.Tensor, residual: torch.Tensor | None = None,
             eps: float = 1e-5, packed: bool = False):
    """The root-mean-square norm of x's rows times weight; with a residual, of
    x + residual, which is returned too: (y, x + residual).  packed: the norm in 8
    bits as well (Packed8, the last of what is returned), for a layer that keeps it."""
    if not isinstance(x, torch.Tensor) or not x.is_cuda or x.dtype not in _DT:
        raise ValueError("x must be an fp32, bf16 or fp16 CUDA tensor")
    dim = weight.numel()
    if weight.dim() != 1 or weight.dtype != x.dtype or weight.device != x.device or (
            dim > 1 and weight.stride(0) != 1):
        raise ValueError("weight must be a vector of x's type, on its device")
    if x.dim() < 1 or x.shape[-1] != dim:
        raise ValueError("x must have rows of %d elements" % dim)
    rows = _rows(x, dim)
    if residual is not None:
        _same("residual", residual, x)
        residual = _rows(residual, dim)
    q = Packed8(rows.shape[0], dim, x.device) if packed else None
    grads = torch.is_grad_enabled() and any(
        t is not None and t.requires_grad for t in (rows, residual, weight))
    y, total, _ = _Norm.apply(rows, residual, weight, float(eps), q, grads)
    out = (y.view(x.shape),) + ((total.view(x.shape),) if total is not None else ()) + (
        (q,) if packed else ())
    return out if len(out) > 1 else out[0]


# --------------------------------------------------- 16-bit products and layers

_ACT = {None: z.ZERO_ACT_NONE, "none": z.ZERO_ACT_NONE, "relu": z.ZERO_ACT_RELU,
        "gelu": z.ZERO_ACT_GELU, "gelu_tanh": z.ZERO_ACT_GELU_TANH, "silu": z.ZERO_ACT_SILU}


def _activation(name) -> int:
    if name not in _ACT:
        raise ValueError("activation must be one of %s" % ", ".join(
            sorted(k for k in _ACT if k)))
    return _ACT[name]


def _operand(name: str, x: torch.Tensor, like: torch.Tensor | None = None) -> torch.Tensor:
    _matrix(name, x)
    if x.dtype == torch.float32:
        raise ValueError("%s must be bf16 or fp16" % name)
    if like is not None and (x.dtype != like.dtype or x.device != like.device):
        raise ValueError("%s must have the other operands' type and device" % name)
    return x


def _place(x):
    return (None, 0) if x is None else (x, _stride(x))


def _workspace(need: int, device):
    return torch.empty(need, dtype=torch.uint8, device=device) if need else None


def matmul(a: torch.Tensor, b: torch.Tensor, a_cols: bool = False, b_cols: bool = False,
           a2: torch.Tensor | None = None, b2: torch.Tensor | None = None,
           bias: torch.Tensor | None = None, activation: str | None = None,
           residual: torch.Tensor | None = None, kept: torch.Tensor | None = None,
           packed: Packed8 | None = None, out: torch.Tensor | None = None,
           accumulate: bool = False) -> torch.Tensor:
    """activation(A B^T + A2 B2^T + bias) + residual, into (or added to) `out` if
    that is given: m by n, of the operands' type or fp32.  A is `a`, m by k, or
    with a_cols its transpose; B is `b`, n by k, or with b_cols its transpose.  The
    sum before the activation also goes to `kept` or `packed`.  Not differentiable:
    the call behind `linear` and `gated`, and the way to a weight's gradient in a
    rank's gradient buffer, matmul(dy, x, True, True, out=grad, accumulate=...)."""
    _operand("a", a)
    _operand("b", b, a)
    m, k = reversed(a.shape) if a_cols else a.shape
    n, kb = reversed(b.shape) if b_cols else b.shape
    if k != kb:
        raise ValueError("the operands must have as many columns")
    if (a2 is None) != (b2 is None):
        raise ValueError("a2 and b2 are given together")
    if a2 is not None:
        _operand("a2", a2, a)
        _operand("b2", b2, a)
        if a2.shape != a.shape or b2.shape != b.shape:
            raise ValueError("a2 and b2 must have the shapes of a and b")
    if out is None:
        if accumulate:
            raise ValueError("there is nothing to add to")
        out = torch.empty(m, n, dtype=a.dtype, device=a.device)
    for name, t in (("out", out), ("residual", residual), ("kept", kept)):
        if t is not None:
            _matrix(name, t)
            if t.shape != (m, n) or t.device != a.device:
                raise ValueError("%s must be %d by %d on %s" % (name, m, n, a.device))
    if out.dtype not in (a.dtype, torch.float32) or (
            residual is not None and residual.dtype != out.dtype):
        raise ValueError("out must be of the operands' type or fp32, and residual of out's")
    if kept is not None and kept.dtype != a.dtype:
        raise ValueError("kept must be of the operands' type")
    if packed is not None and ((packed.rows, packed.cols) != (m, n)
                               or packed.q.device != a.device):
        raise ValueError("packed must be %d by %d on %s" % (m, n, a.device))
    if bias is not None and (bias.shape != (n,) or bias.dtype != a.dtype
                             or bias.device != a.device or (n > 1 and bias.stride(0) != 1)):
        raise ValueError("bias must be a vector of %d elements of the operands' type" % n)
    _product(a, b, a_cols, b_cols, a2, b2, bias, _activation(activation), residual, kept,
             packed.q if packed is not None else None, out, accumulate, m, n, k)
    _written(out, kept)
    return out


def _product(a, b, a_cols, b_cols, a2, b2, bias, act, residual, kept, kept_q, out, accumulate, m,
             n, k):
    pa, pb, pa2, pb2 = _place(a), _place(b), _place(a2), _place(b2)
    with torch.cuda.device(a.device):
        need = z.zero_matmul_workspace(pa[0], a_cols, pa[1], pb[0], b_cols, pb[1], *pa2, *pb2, m,
                                       n, k)
        z.zero_matmul(pa[0], a_cols, pa[1], pb[0], b_cols, pb[1], *pa2, *pb2, _DT[a.dtype], m, n,
                      k, bias, act, *_place(residual), *_place(kept), kept_q, out, _DT[out.dtype],
                      _stride(out), accumulate, _workspace(need, a.device), need)
    return out


def _empty(x, rows, cols):
    return torch.empty(rows, cols, dtype=x.dtype, device=x.device)


def _keep_input(x, keep8):
    """What is kept of a layer's input: itself, or its 8-bit form, which an
    earlier norm may have made."""
    if keep8 is False:
        return x
    return (keep8 if isinstance(keep8, Packed8) else pack8(x)).q


class _Dense(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, weight, bias, residual, act, keep8, grads):
        ctx.set_materialize_grads(False)
        (m, k), n = x.shape, weight.shape[0]
        need_x, need_w, need_b = (grads and v for v in ctx.needs_input_grad[:3])
        kept = kept_q = None
        if act != z.ZERO_ACT_NONE and (need_x or need_w or need_b):
            if keep8 is False:
                kept = _empty(x, m, n)
            else:
                kept_q = Packed8(m, n, x.device).q
        out = _product(x, weight, False, False, None, None, bias, act, residual, kept, kept_q,
                       _empty(x, m, n), False, m, n, k)
        ctx.shape, ctx.act, ctx.packed = (m, n, k), act, keep8 is not False
        link = None
        if grads:
            link = x.new_empty(0)
            ctx.save_for_backward(_keep_input(x, keep8) if need_w else None,
                                  weight if need_x else None, kept if kept_q is None else kept_q,
                                  link)
        ctx.dtype, ctx.device = x.dtype, x.device
        return out, link

    @staticmethod
    def backward(ctx, dy, _):
        if dy is None:
            return (None,) * 7
        x, weight, kept, link = ctx.saved_tensors
        m, n, k = ctx.shape
        need_x, need_w, need_b, need_r = ctx.needs_input_grad[:4]
        given = dy
        dy = _gradient(dy)
        dx = dw = db = None
        with torch.cuda.device(ctx.device):
            dz = dy
            if need_b or (ctx.act != z.ZERO_ACT_NONE and (need_x or need_w)):
                if ctx.act != z.ZERO_ACT_NONE:
                    dz = torch.empty(m, n, dtype=ctx.dtype, device=ctx.device)
                if need_b:
                    db = torch.empty(n, dtype=ctx.dtype, device=ctx.device)
                need = z.zero_activation_grad_workspace(m, n) if need_b else 0
                dt = _DT[ctx.dtype]
                z.zero_activation_grad(
                    dy, _stride(dy), None if ctx.packed else kept, n, kept if ctx.packed else None,
                    ctx.act, dt, m, n, None if dz is dy else dz, n, db, dt, False,
                    _workspace(need, ctx.device), need)
            if need_x:
                dx = _product(dz, weight, False, True, None, None, None, 0, None, None, None,
                              _empty(dz, m, k), False, m, k, n)
            if need_w:
                if ctx.packed:
                    x = _unpacked(x, m, k, ctx.dtype)
                dw = _product(dz, x, True, True, None, None, None, 0, None, None, None,
                              _empty(dz, n, k), False, n, k, m)
        dx, dw, db = _last("linear", (dx, dw, db), given, link)
        return dx, dw, db, given if need_r else None, None, None, None


def _weight(name, w, x):
    _operand(name, w, x)
    if w.shape[1] != x.shape[1]:
        raise ValueError("%s must have rows of %d elements" % (name, x.shape[1]))


def _check_keep8(keep8, rows):
    if isinstance(keep8, Packed8):
        if (keep8.rows, keep8.cols) != tuple(rows.shape) or keep8.q.device != rows.device:
            raise ValueError("keep8 must be x's 8-bit form")
        return keep8
    return bool(keep8)


def linear(x: torch.Tensor, weight: torch.Tensor, bias: torch.Tensor | None = None,
           activation: str | None = None, residual: torch.Tensor | None = None,
           keep8: bool | Packed8 = False) -> torch.Tensor:
    """activation(x weight^T + bias) + residual in bf16 or fp16, weight [n, k], the
    sums in fp32 and one rounding at the end.  The gradients are those at what is
    kept: x and, with an activation, its argument, in x's type or, with keep8, in 8 bits
    (keep8 may be x's Packed8 itself, as rms_norm gives it)."""
    if not isinstance(x, torch.Tensor) or x.dim() < 1 or not isinstance(weight, torch.Tensor) or (
            weight.dim() != 2) or x.shape[-1] != weight.shape[1]:
        raise ValueError("x must have rows as long as weight's")
    n, k = weight.shape
    rows = _operand("x", _rows(x, k))
    _weight("weight", weight, rows)
    if bias is not None and (bias.shape != (n,) or bias.dtype != x.dtype or
                             bias.device != x.device or (n > 1 and bias.stride(0) != 1)):
        raise ValueError("bias must be a vector of %d elements of x's type, on its device" % n)
    shape = (*x.shape[:-1], n)
    if residual is not None:
        if residual.shape != shape or residual.dtype != x.dtype or residual.device != x.device:
            raise ValueError("residual must have the result's shape, type and device")
        residual = _rows(residual, n)
    grads = torch.is_grad_enabled() and any(
        t is not None and t.requires_grad for t in (rows, weight, bias, residual))
    return _Dense.apply(rows, weight, bias, residual, _activation(activation),
                        _check_keep8(keep8, rows), grads)[0].view(shape)


class _Gated(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, w_gate, w_up, act, keep8, grads):
        ctx.set_materialize_grads(False)
        (m, k), n = x.shape, w_gate.shape[0]
        gate = up = gate_q = up_q = None
        if grads and keep8 is False:
            gate, up = _empty(x, m, n), _empty(x, m, n)
        elif grads:
            gate_q, up_q = Packed8(m, n, x.device).q, Packed8(m, n, x.device).q
        h = _empty(x, m, n)
        with torch.cuda.device(x.device):
            places = *_place(x), *_place(w_gate), *_place(w_up)
            need = z.zero_gated_workspace(*places, m, n, k)
            z.zero_gated(*places, _DT[x.dtype], m, n, k, act, gate, up, n, gate_q, up_q, h, n,
                         _workspace(need, x.device), need)
        ctx.shape, ctx.act, ctx.packed = (m, n, k), act, keep8 is not False
        link = None
        if grads:
            link = x.new_empty(0)
            need_x, need_g, need_u = ctx.needs_input_grad[:3]
            ctx.save_for_backward(_keep_input(x, keep8) if need_g or need_u else None,
                                  w_gate if need_x else None, w_up if need_x else None,
                                  *((gate_q, up_q) if ctx.packed else (gate, up)), link)
        ctx.dtype, ctx.device = x.dtype, x.device
        return h, link

    @staticmethod
    def backward(ctx, dh, _):
        if dh is None:
            return (None,) * 6
        x, w_gate, w_up, gate, up, link = ctx.saved_tensors
        m, n, k = ctx.shape
        need_x, need_g, need_u = ctx.needs_input_grad[:3]
        given = dh
        dh = _gradient(dh)
        dx = dwg = dwu = None
        with torch.cuda.device(ctx.device):
            dg, du = _empty(dh, m, n), _empty(dh, m, n)
            kept = (None, None, n, gate, up) if ctx.packed else (gate, up, n, None, None)
            z.zero_gated_grad(dh, _stride(dh), *kept, ctx.act, _DT[ctx.dtype], m, n, dg, du, n)
            if need_x:
                dx = _product(dg, w_gate, False, True, du, w_up, None, 0, None, None, None,
                              _empty(dh, m, k), False, m, k, n)
            if x is not None and ctx.packed:
                x = _unpacked(x, m, k, ctx.dtype)
            if need_g:
                dwg = _product(dg, x, True, True, None, None, None, 0, None, None, None,
                               _empty(dh, n, k), False, n, k, m)
            if need_u:
                dwu = _product(du, x, True, True, None, None, None, 0, None, None, None,
                               _empty(dh, n, k), False, n, k, m)
        return (*_last("gated", (dx, dwg, dwu), given, link), None, None, None)


def gated(x: torch.Tensor, w_gate: torch.Tensor, w_up: torch.Tensor,
          activation: str | None = "silu", keep8: bool | Packed8 = False) -> torch.Tensor:
    """activation(x w_gate^T) * (x w_up^T) in bf16 or fp16, both weights [n, k], in
    one pass over x.  The gradients are those at what is kept: x and both projections,
    in x's type or, with keep8, in 8 bits (see linear)."""
    if not isinstance(x, torch.Tensor) or x.dim() < 1 or not isinstance(
            w_gate, torch.Tensor) or w_gate.dim() != 2 or x.shape[-1] != w_gate.shape[1]:
        raise ValueError("x must have rows as long as the weights'")
    n, k = w_gate.shape
    rows = _operand("x", _rows(x, k))
    _weight("w_gate", w_gate, rows)
    _weight("w_up", w_up, rows)
    if w_up.shape != w_gate.shape:
        raise ValueError("the weights must have one shape")
    grads = torch.is_grad_enabled() and any(t.requires_grad for t in (rows, w_gate, w_up))
    return _Gated.apply(rows, w_gate, w_up, _activation(activation), _check_keep8(keep8, rows),
                        grads)[0].view(*x.shape[:-1], n)
